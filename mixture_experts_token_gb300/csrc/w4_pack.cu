// 4-bit weights with group scales: quantising, laying out for the products
// (w4.cuh has the layout) and expanding again.  Work of loading a model, not
// of a step: each kernel reads its input once and writes its output once
// (the quantiser reads a group twice, the second time from the caches).
// Measured, 256 bf16 matrices of 7168 x 2048 in groups of 128: quantise 6.0 ms
// and expand 7.5 ms, 8.4 ms with zero points (1.4 ms of bytes at 6.8 TB/s),
// pack 2.7 ms (0.57 ms).  Only packing was tuned: a thread of the quantiser
// loads one value at a time, and the expander reads a word of codes anew for
// each of its eight nibbles.
#include <cuda_bf16.h>
#include <math.h>

#include <limits>

#include "w4.cuh"

namespace moe {
namespace {

using namespace w4;

constexpr int kThreads = 256;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
__device__ __forceinline__ void from_float(float v, float* p) { *p = v; }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16* p) {
  *p = __float2bfloat16(v);
}

// A thread per (matrix, group, column): its group's scale (and zero), then
// its codes.  The scale is rounded to bf16 first and the codes are nearest
// to the weights under the rounded scale.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T* __restrict__ w, int n_mats, Layout l,
                    uint8_t* __restrict__ codes,
                    __nv_bfloat16* __restrict__ scales,
                    uint8_t* __restrict__ zeros) {
  const int G = l.groups();
  const long long total = static_cast<long long>(n_mats) * G * l.N;
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) +
                     threadIdx.x;
       i < total; i += static_cast<long long>(gridDim.x) * kThreads) {
    const int n = static_cast<int>(i % l.N);
    const long long mg = i / l.N;
    const int g = static_cast<int>(mg % G);
    const long long m = mg / G;
    const int k0 = g * l.group, k1 = min(l.K, k0 + l.group);
    const T* src = w + m * l.K * l.N + n;
    float lo = 0.0f, hi = 0.0f;  // the range always holds zero
    for (int k = k0; k < k1; ++k) {
      const float v = to_float(src[static_cast<long long>(k) * l.N]);
      lo = fminf(lo, v);
      hi = fmaxf(hi, v);
    }
    const float span = l.zeros ? (hi - lo) / 15.0f : fmaxf(-lo, hi) / 7.0f;
    const __nv_bfloat16 sb = __float2bfloat16(span);
    const float s = __bfloat162float(sb);
    const float z =
        !l.zeros ? 8.0f
        : s > 0.0f ? fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f)
                   : 0.0f;
    scales[i] = sb;
    if (l.zeros) zeros[i] = static_cast<uint8_t>(z);
    uint8_t* dst = codes + m * (l.K / 2) * l.N + n;
    for (int k = k0; k < k1; k += 2) {
      int q[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float v = to_float(src[static_cast<long long>(k + j) * l.N]);
        const float c = s > 0.0f ? rintf(v / s) + z : z;
        q[j] = static_cast<int>(fminf(fmaxf(c, 0.0f), 15.0f));
      }
      dst[static_cast<long long>(k / 2) * l.N] =
          static_cast<uint8_t>(q[0] | (q[1] << 4));
    }
  }
}

// Row and column of nibble i of word s of lane `lane` within a tile.
__device__ __forceinline__ int nibble_k(int lane, int s, int i) {
  return 16 * s + 2 * (lane & 3) + ((i >> 2) & 1) + 4 * (i & 2);
}
__device__ __forceinline__ int nibble_n(int lane, int i) {
  return (lane >> 2) + 8 * (i & 1);
}
// Bytes from a record's start to a tile of codes.
__device__ __forceinline__ long long code_at(const Layout& l, int tile) {
  constexpr int kPer = kStepK / kTileK;
  return l.step_at(tile / kPer) + tile % kPer * kTileBytes;
}

// A CTA packs four records (64 columns) of a matrix, 128 rows at a time:
// codes come in rows of 64 bytes to shared memory and leave as whole words.
// grid.y strides over matrices.  256 matrices of 7168 x 2048, 1.9 GB of
// codes: 2.7 ms, and about 6 ms with a byte load for every code.
constexpr int kPackRecords = 4;
constexpr int kPackCols = kPackRecords * kTileN;
constexpr int kPackK = 2 * kTileK;
__global__ void __launch_bounds__(kThreads)
    pack_kernel(const uint8_t* __restrict__ codes,
                const __nv_bfloat16* __restrict__ scales,
                const uint8_t* __restrict__ zeros, int n_mats, Layout l,
                bool wide, char* __restrict__ packed) {
  // written as words; rows 4 bytes past 64: neighbouring rows start in
  // neighbouring banks
  __shared__ __align__(4) uint8_t rows[kPackK / 2][kPackCols + 4];
  const int n0 = blockIdx.x * kPackCols, G = l.groups();
  const int E = kStepK / l.group;  // groups of a step
  const int records = min(kPackRecords, l.tiles_n() - kPackRecords *
                                            static_cast<int>(blockIdx.x));
  for (long long m = blockIdx.y; m < n_mats; m += gridDim.y) {
    const uint8_t* c = codes + m * (l.K / 2) * l.N;
    const __nv_bfloat16* sc = scales + m * G * l.N;
    const uint8_t* zp = l.zeros ? zeros + m * G * l.N : nullptr;
    char* rec0 = packed + m * l.matrix() +
                 static_cast<long long>(blockIdx.x) * kPackRecords *
                     l.record();
    for (int k0 = 0; k0 < l.K; k0 += kPackK) {
      __syncthreads();
      const int r = threadIdx.x / 4, q = threadIdx.x % 4 * 16;
      uint32_t v[4] = {0, 0, 0, 0};
      if (2 * r + k0 < l.K) {
        const uint8_t* src = c + (k0 / 2 + r) * static_cast<long long>(l.N) +
                             n0 + q;
        if (wide && n0 + q + 16 <= l.N) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(src));
          v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
        } else {
          for (int i = 0; i < 16; ++i)
            if (n0 + q + i < l.N)
              v[i / 4] |= static_cast<uint32_t>(src[i]) << (8 * (i % 4));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint32_t*>(&rows[r][q + 4 * i]) = v[i];
      __syncthreads();
      const int tiles = min(2, l.tiles_k() - k0 / kTileK);
      for (int i = threadIdx.x; i < records * tiles * 128; i += kThreads) {
        const int rec = i / (tiles * 128), tile = i / 128 % tiles;
        const int lane = (i >> 2) & 31, s = i & 3;
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int kt = tile * kTileK + nibble_k(lane, s, j), k = k0 + kt;
          const int col = rec * kTileN + nibble_n(lane, j), n = n0 + col;
          uint32_t code = l.zeros ? 0 : 8;
          if (n < l.N) {
            if (k < l.K) {
              const uint32_t b = rows[kt / 2][col];
              code = k & 1 ? b >> 4 : b & 15;
            } else if (l.zeros) {
              // the stored zero of k's group: 0 past the last group
              const int g = k / l.group;
              code = g < G ? zp[static_cast<long long>(g) * l.N + n] & 15 : 0;
            }
          }
          word |= code << (4 * j);
        }
        *reinterpret_cast<uint32_t*>(rec0 + rec * l.record() +
                                     code_at(l, k0 / kTileK + tile) +
                                     (i & 127) * 4) = word;
      }
    }
    for (int i = threadIdx.x; i < records * l.steps() * 16 * E;
         i += kThreads) {
      const int rec = i / (l.steps() * 16 * E);
      const int at = i - rec * (l.steps() * 16 * E);
      const int step = at / (16 * E), j = at % (16 * E);
      const int n = n0 + rec * kTileN + j / (2 * E) + 8 * (j & 1);
      const int g = step * E + j / 2 % E;
      const bool in = n < l.N && g < G;
      const long long from = static_cast<long long>(g) * l.N + n;
      char* so = rec0 + rec * l.record() + l.scales_at(step);
      reinterpret_cast<__nv_bfloat16*>(so)[j] =
          in ? sc[from] : __float2bfloat16(0.0f);
      if (l.zeros) so[32 * E + j] = in ? zp[from] & 15 : 0;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const char* __restrict__ packed, int n_mats, Layout l,
                      T* __restrict__ w) {
  const int n0 = blockIdx.x * kTileN, E = kStepK / l.group;
  for (long long m = blockIdx.y; m < n_mats; m += gridDim.y) {
    const char* rec = packed + m * l.matrix() + blockIdx.x * l.record();
    T* dst = w + m * l.K * l.N;
    for (int i = threadIdx.x; i < l.K * kTileN; i += kThreads) {
      const int k = i / kTileN, col = i % kTileN, n = n0 + col;
      if (n >= l.N) continue;
      const int r = k % kTileK;
      const int lane = (col & 7) * 4 + ((r >> 1) & 3), s = r >> 4;
      const int j = (col >> 3) + 2 * ((r >> 3) & 1) + 4 * (r & 1);
      const uint32_t v = *reinterpret_cast<const uint32_t*>(
          rec + code_at(l, k / kTileK) + lane * 16 + s * 4);
      const uint32_t q = v >> (4 * j) & 15;
      const char* so = rec + l.scales_at(k / kStepK);
      const int at = ((col & 7) * E + k % kStepK / l.group) * 2 + (col >> 3);
      const int z = l.zeros ? so[32 * E + at] : 8;
      from_float(static_cast<float>(static_cast<int>(q) - z) *
                     __bfloat162float(
                         reinterpret_cast<const __nv_bfloat16*>(so)[at]),
                 dst + static_cast<long long>(k) * l.N + n);
    }
  }
}

bool shape_ok(int n, int K, int N) {
  return n >= 0 && K >= 2 && K % 2 == 0 && N >= 1 && K <= (1 << 20) &&
         N <= (1 << 20);
}
dim3 record_grid(const Layout& l, int n) {
  return dim3(l.tiles_n(), n < 4096 ? n : 4096);
}
// scales are read and written one by one: their natural alignment is enough
bool ok_scales(const void* p) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 1) == 0;
}
moe_status_t launched() {
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;
using namespace moe::w4;

extern "C" {

size_t moe_w4_bytes(const moe_w4_t* opt, int32_t n, int32_t K, int32_t N) {
  if (!w4::options_ok(opt) || !shape_ok(n, K, N)) return 0;
  return static_cast<size_t>(layout(*opt, K, N).matrix()) * n;
}

moe_status_t moe_w4_quantize(const moe_w4_t* opt, int32_t n, int32_t K,
                             int32_t N, moe_dtype_t dtype, const void* w,
                             uint8_t* codes, void* scales, uint8_t* zeros,
                             moe_stream_t stream) {
  if (!w4::options_ok(opt) || !shape_ok(n, K, N) ||
      (dtype != MOE_F32 && dtype != MOE_BF16))
    return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!ok_ptr(w, true) || codes == nullptr || !ok_scales(scales) ||
      (zeros != nullptr) != (opt->zero_points != 0))
    return MOE_ERR_INVALID_ARG;
  const Layout l = layout(*opt, K, N);
  const long long total = static_cast<long long>(n) * l.groups() * N;
  const unsigned grid = static_cast<unsigned>(
      std::min<long long>((total + kThreads - 1) / kThreads, 1 << 20));
  __nv_bfloat16* sc = static_cast<__nv_bfloat16*>(scales);
  if (dtype == MOE_F32)
    quantize_kernel<<<grid, kThreads, 0, stream>>>(
        static_cast<const float*>(w), n, l, codes, sc, zeros);
  else
    quantize_kernel<<<grid, kThreads, 0, stream>>>(
        static_cast<const __nv_bfloat16*>(w), n, l, codes, sc, zeros);
  return launched();
}

moe_status_t moe_w4_pack(const moe_w4_t* opt, int32_t n, int32_t K, int32_t N,
                         const uint8_t* codes, const void* scales,
                         const uint8_t* zeros, void* packed,
                         moe_stream_t stream) {
  if (!w4::options_ok(opt) || !shape_ok(n, K, N)) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (codes == nullptr || !ok_scales(scales) || !ok_ptr(packed, true) ||
      (zeros != nullptr) != (opt->zero_points != 0))
    return MOE_ERR_INVALID_ARG;
  const Layout l = layout(*opt, K, N);
  const dim3 grid((l.tiles_n() + kPackRecords - 1) / kPackRecords,
                  n < 4096 ? n : 4096);
  pack_kernel<<<grid, kThreads, 0, stream>>>(
      codes, static_cast<const __nv_bfloat16*>(scales), zeros, n, l,
      aligned16(codes) && N % 16 == 0, static_cast<char*>(packed));
  return launched();
}

moe_status_t moe_w4_dequantize(const moe_w4_t* opt, int32_t n, int32_t K,
                               int32_t N, const void* packed,
                               moe_dtype_t dtype, void* w,
                               moe_stream_t stream) {
  if (!w4::options_ok(opt) || !shape_ok(n, K, N) ||
      (dtype != MOE_F32 && dtype != MOE_BF16))
    return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!ok_ptr(packed, true) || !ok_ptr(w, true)) return MOE_ERR_INVALID_ARG;
  const Layout l = layout(*opt, K, N);
  const char* p = static_cast<const char*>(packed);
  if (dtype == MOE_F32)
    dequantize_kernel<<<record_grid(l, n), kThreads, 0, stream>>>(
        p, n, l, static_cast<float*>(w));
  else
    dequantize_kernel<<<record_grid(l, n), kThreads, 0, stream>>>(
        p, n, l, static_cast<__nv_bfloat16*>(w));
  return launched();
}

}  // extern "C"
