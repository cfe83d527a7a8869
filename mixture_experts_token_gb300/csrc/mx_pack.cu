// Microscaled 4-bit numbers (mx.cuh): quantising rows and weight matrices,
// laying matrices out for the products, and expanding both again.  Each
// kernel reads its input once and writes its output once, so bytes bound it.
#include "launch.cuh"
#include "mx.cuh"

namespace moe {
namespace {

using namespace mx;

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(const float (&v)[8], float* p) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(const float (&v)[8],
                                       __nv_bfloat16* p) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight values of a row a thread, so a block is two or four lanes.
template <int BLOCK, typename T>
__global__ void __launch_bounds__(kThreads)
    quantize_rows_kernel(const T* __restrict__ x, long long pieces, int K,
                         float r, uint8_t* __restrict__ codes,
                         uint8_t* __restrict__ scales) {
  constexpr int kLanes = BLOCK / 8;
  launch::wait_for_previous();
  launch::let_next_start();
  const int per_row = K / 8, sr = scale_row(K, BLOCK);
  // pieces is a multiple of the lanes of a block: they leave together
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) +
                     threadIdx.x;
       i < pieces; i += static_cast<long long>(gridDim.x) * kThreads) {
    float v[8];
    load8(x + i * 8, v);
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (BLOCK == 16) v[j] *= r;
      most = max(most, __float_as_uint(v[j]) & 0x7fffffffu);
    }
    const uint32_t mask =
        ((1u << kLanes) - 1) << (threadIdx.x & 31 & ~(kLanes - 1));
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1)
      most = max(most, __shfl_xor_sync(mask, most, o));
    const Block b = block_scale<BLOCK>(most);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = over_scale<BLOCK>(v[j], b);
    reinterpret_cast<uint32_t*>(codes)[i] = encode8(v);
    if (threadIdx.x % kLanes == 0) {
      const long long row = i / per_row;
      const int at = static_cast<int>(i - row * per_row) / kLanes;
      uint8_t* s = scales + row * sr;
      s[at] = static_cast<uint8_t>(b.byte);
      if (at == K / BLOCK - 1)
        for (int j = at + 1; j < sr; ++j) s[j] = 0;
    }
  }
}

template <int BLOCK, typename T>
__global__ void __launch_bounds__(kThreads)
    dequantize_rows_kernel(const uint8_t* __restrict__ codes,
                           const uint8_t* __restrict__ scales,
                           long long pieces, int K, float scale,
                           T* __restrict__ x) {
  const int per_row = K / 8, sr = scale_row(K, BLOCK);
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) +
                     threadIdx.x;
       i < pieces; i += static_cast<long long>(gridDim.x) * kThreads) {
    const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(codes) + i);
    const long long row = i / per_row;
    const int at = static_cast<int>(i - row * per_row) / (BLOCK / 8);
    const float s = scale_value<BLOCK>(__ldg(scales + row * sr + at));
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = decode(c >> (4 * j) & 15) * s;  // exact
      if (BLOCK == 16) v[j] *= scale;
    }
    store8(v, x + i * 8);
  }
}

// A weight matrix w [K, N] becomes N rows of codes: 64 columns and 256 of K
// at a time through shared memory, read a row of w and written a row of codes
// at a time.  A thread takes 32 of K of one column.
constexpr int kTurnN = 64;
template <int BLOCK, typename T>
__global__ void __launch_bounds__(kThreads)
    quantize_weights_kernel(const T* __restrict__ w,
                            const float* __restrict__ scale, int n_mats,
                            int K, int N, uint8_t* __restrict__ codes,
                            uint8_t* __restrict__ scales) {
  // an odd number of words a row: eight of k apart is four banks apart
  extern __shared__ char raw[];
  constexpr int kPitch = kTurnN + 4 / sizeof(T);
  T* tile = reinterpret_cast<T*>(raw);
  const int n0 = blockIdx.x * kTurnN, k0 = blockIdx.y * kStageK;
  const int sr = scale_row(K, BLOCK);
  for (long long m = blockIdx.z; m < n_mats; m += gridDim.z) {
    const float r = BLOCK == 16 && scale ? __frcp_rn(scale[m]) : 1.0f;
    __syncthreads();
    for (int i = threadIdx.x; i < kStageK * kTurnN; i += kThreads) {
      const int k = i / kTurnN, n = i % kTurnN;
      if (k0 + k < K && n0 + n < N)
        tile[k * kPitch + n] = w[(m * K + k0 + k) * N + n0 + n];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kTurnN * (kStageK / 32); i += kThreads) {
      const int n = i / (kStageK / 32), k = i % (kStageK / 32) * 32;
      if (n0 + n >= N || k0 + k >= K) continue;
      const long long row = m * N + n0 + n;
      uint32_t out[4];
#pragma unroll
      for (int h = 0; h < 32 / BLOCK; ++h) {
        float v[BLOCK];
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < BLOCK; ++j) {
          v[j] = to_float(tile[(k + h * BLOCK + j) * kPitch + n]) * r;
          most = max(most, __float_as_uint(v[j]) & 0x7fffffffu);
        }
        const Block b = block_scale<BLOCK>(most);
#pragma unroll
        for (int j = 0; j < BLOCK / 8; ++j) {
          float q[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) q[e] = over_scale<BLOCK>(v[8 * j + e], b);
          out[h * (BLOCK / 8) + j] = encode8(q);
        }
        const int at = (k0 + k) / BLOCK + h;
        uint8_t* s = scales + row * sr;
        s[at] = static_cast<uint8_t>(b.byte);
        if (at == K / BLOCK - 1)
          for (int j = at + 1; j < sr; ++j) s[j] = 0;
      }
      *reinterpret_cast<uint4*>(codes + row * (K / 2) + (k0 + k) / 2) =
          make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
}

// Rows of codes and scales to records, a CTA for each.
template <int BLOCK>
__global__ void __launch_bounds__(kThreads)
    pack_kernel(const uint8_t* __restrict__ codes,
                const uint8_t* __restrict__ scales, int n_mats, Layout l,
                char* __restrict__ packed) {
  constexpr int kTiles = scale_tiles(BLOCK);
  const int stage = blockIdx.x, n0 = blockIdx.y * kTileN;
  const int sr = scale_row(l.K, BLOCK), groups = l.K / BLOCK;
  for (long long m = blockIdx.z; m < n_mats; m += gridDim.z) {
    char* rec = packed + m * l.matrix() + blockIdx.y * l.tile() +
                static_cast<long long>(stage) * record_bytes(BLOCK);
    const long long row0 = m * l.N + n0;
    for (int i = threadIdx.x; i < kTileN * 8; i += kThreads) {
      const int r = i / 8, p = i % 8, at = stage * (kStageK / 2) + p * 16;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (n0 + r < l.N && at < l.K / 2)
        v = __ldg(reinterpret_cast<const uint4*>(codes + (row0 + r) *
                                                             (l.K / 2) +
                                                 at));
      *reinterpret_cast<uint4*>(rec + r * 128 + ((p ^ (r & 7)) << 4)) = v;
    }
    for (int i = threadIdx.x; i < kTileN * kTiles; i += kThreads) {
      const int r = i / kTiles, j = i % kTiles;
      const int at = (stage * kTiles + j) * 4;
      uint32_t v = 0;
      if (n0 + r < l.N && at < groups) {
        v = __ldg(reinterpret_cast<const uint32_t*>(scales + (row0 + r) * sr +
                                                    at));
        // what lies behind the row's last scale counts as zero
        if (groups - at < 4) v &= (1u << (8 * (groups - at))) - 1;
      }
      *reinterpret_cast<uint32_t*>(rec + kCodeBytes + j * kScaleTile +
                                   r % 32 * 16 + r / 32 * 4) = v;
    }
  }
}

// Records to w [K, N], a CTA for each: a thread expands eight of K of a
// column, and the 128 columns of a row of w are written side by side.
template <int BLOCK, typename T>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const char* __restrict__ packed,
                      const float* __restrict__ scale, int n_mats, Layout l,
                      T* __restrict__ w) {
  __shared__ __align__(16) char rec[record_bytes(BLOCK)];
  const int stage = blockIdx.x, n0 = blockIdx.y * kTileN;
  for (long long m = blockIdx.z; m < n_mats; m += gridDim.z) {
    const char* src = packed + m * l.matrix() + blockIdx.y * l.tile() +
                      static_cast<long long>(stage) * record_bytes(BLOCK);
    __syncthreads();
    for (int i = threadIdx.x; i < record_bytes(BLOCK) / 16; i += kThreads)
      reinterpret_cast<uint4*>(rec)[i] =
          __ldg(reinterpret_cast<const uint4*>(src) + i);
    __syncthreads();
    const float t = BLOCK == 16 && scale ? scale[m] : 1.0f;
    for (int i = threadIdx.x; i < kTileN * (kStageK / 8); i += kThreads) {
      const int r = i % kTileN, p = i / kTileN;  // column, eight of k
      const int k = stage * kStageK + p * 8;
      if (n0 + r >= l.N || k >= l.K) continue;
      const uint32_t c = *reinterpret_cast<const uint32_t*>(
          rec + r * 128 + ((p / 4 ^ (r & 7)) << 4) + p % 4 * 4);
      const int g = p * 8 / BLOCK;
      const float s = scale_value<BLOCK>(static_cast<uint8_t>(
          rec[kCodeBytes + g / 4 * kScaleTile + r % 32 * 16 + r / 32 * 4 +
              g % 4]));
      T* out = w + (m * l.K + k) * l.N + n0 + r;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = decode(c >> (4 * j) & 15) * s;
        if (BLOCK == 16) v *= t;
        put(out + static_cast<long long>(j) * l.N, v);
      }
    }
  }
}

bool dtype_ok(moe_dtype_t d) { return d == MOE_F32 || d == MOE_BF16; }
bool matrix_ok(int n, int K, int N) {
  return n >= 0 && length_ok(K) && N >= 1 && N <= (1 << 20);
}
bool rows_ok(int R, int K) { return R >= 0 && length_ok(K); }
moe_status_t status_of(cudaError_t e) {
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
moe_status_t launched() { return status_of(cudaGetLastError()); }
unsigned row_grid(long long pieces) {
  return static_cast<unsigned>(
      std::min<long long>((pieces + kThreads - 1) / kThreads, 1 << 20));
}
dim3 record_grid(const Layout& l, int n) {
  return dim3(l.stages(), l.tiles_n(), n < 4096 ? n : 4096);
}

template <int BLOCK, typename T>
cudaError_t quantize_weights(int n, int K, int N, const void* w,
                             const float* scale, uint8_t* codes,
                             uint8_t* scales, cudaStream_t s) {
  constexpr auto kernel = quantize_weights_kernel<BLOCK, T>;
  launch::Device d;
  cudaError_t e = launch::device(&d);
  if (e == cudaSuccess) e = launch::allow_shared<kernel>(d);
  if (e != cudaSuccess) return e;
  const dim3 grid((N + kTurnN - 1) / kTurnN, (K + kStageK - 1) / kStageK,
                  n < 4096 ? n : 4096);
  const int bytes = kStageK * (kTurnN * sizeof(T) + 4);
  kernel<<<grid, kThreads, bytes, s>>>(static_cast<const T*>(w), scale, n, K,
                                       N, codes, scales);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_rows(int block, int R, int K, moe_dtype_t dtype,
                           const void* x, float scale, uint8_t* codes,
                           uint8_t* scales, cudaStream_t s) {
  const long long pieces = static_cast<long long>(R) * (K / 8);
  const float r = 1.0f / scale;
  const unsigned grid = row_grid(pieces);
#define MOE_MX_ROWS(B, T)                                                   \
  return launch::overlapping(quantize_rows_kernel<B, T>, grid, kThreads, 0, \
                             s, static_cast<const T*>(x), pieces, K, r,     \
                             codes, scales)
  if (block == 16) {
    if (dtype == MOE_F32) MOE_MX_ROWS(16, float);
    MOE_MX_ROWS(16, __nv_bfloat16);
  }
  if (dtype == MOE_F32) MOE_MX_ROWS(32, float);
  MOE_MX_ROWS(32, __nv_bfloat16);
#undef MOE_MX_ROWS
}

}  // namespace moe

using namespace moe;
using namespace moe::mx;

// Calls f<BLOCK, T> of the call's block and type.
#define MOE_MX_PICK(f, ...)                                         \
  (opt->block == 16                                                 \
       ? (dtype == MOE_F32 ? f<16, float> __VA_ARGS__               \
                           : f<16, __nv_bfloat16> __VA_ARGS__)      \
       : (dtype == MOE_F32 ? f<32, float> __VA_ARGS__               \
                           : f<32, __nv_bfloat16> __VA_ARGS__))

extern "C" {

size_t moe_mx_bytes(const moe_mx_t* opt, int32_t n, int32_t K, int32_t N) {
  if (!mx::options_ok(opt) || !matrix_ok(n, K, N)) return 0;
  return static_cast<size_t>(Layout{K, N, opt->block}.matrix()) * n;
}

int32_t moe_mx_scale_row(const moe_mx_t* opt, int32_t K) {
  return mx::options_ok(opt) && length_ok(K) ? scale_row(K, opt->block) : 0;
}

moe_status_t moe_mx_quantize_rows(const moe_mx_t* opt, int32_t R, int32_t K,
                                  moe_dtype_t dtype, const void* x,
                                  float scale, uint8_t* codes,
                                  uint8_t* scales, moe_stream_t stream) {
  if (!mx::options_ok(opt) || !rows_ok(R, K) || !dtype_ok(dtype) ||
      !scale_ok(opt->block, scale))
    return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (!ok_ptr(x, true) || !ok_ptr(codes, true) || !ok_ptr(scales, false))
    return MOE_ERR_INVALID_ARG;
  return status_of(launch_mx_rows(opt->block, R, K, dtype, x, scale, codes,
                                  scales, stream));
}

moe_status_t moe_mx_dequantize_rows(const moe_mx_t* opt, int32_t R, int32_t K,
                                    const uint8_t* codes,
                                    const uint8_t* scales, float scale,
                                    moe_dtype_t dtype, void* x,
                                    moe_stream_t stream) {
  if (!mx::options_ok(opt) || !rows_ok(R, K) || !dtype_ok(dtype) ||
      !scale_ok(opt->block, scale))
    return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (!ok_ptr(codes, true) || !ok_ptr(scales, false) || !ok_ptr(x, true))
    return MOE_ERR_INVALID_ARG;
  const long long pieces = static_cast<long long>(R) * (K / 8);
#define MOE_MX_ROWS(B, T)                                             \
  dequantize_rows_kernel<B, T><<<row_grid(pieces), kThreads, 0, stream>>>( \
      codes, scales, pieces, K, scale, static_cast<T*>(x))
  if (opt->block == 16) {
    if (dtype == MOE_F32)
      MOE_MX_ROWS(16, float);
    else
      MOE_MX_ROWS(16, __nv_bfloat16);
  } else if (dtype == MOE_F32) {
    MOE_MX_ROWS(32, float);
  } else {
    MOE_MX_ROWS(32, __nv_bfloat16);
  }
#undef MOE_MX_ROWS
  return launched();
}

moe_status_t moe_mx_quantize(const moe_mx_t* opt, int32_t n, int32_t K,
                             int32_t N, moe_dtype_t dtype, const void* w,
                             const float* scale, uint8_t* codes,
                             uint8_t* scales, moe_stream_t stream) {
  if (!mx::options_ok(opt) || !matrix_ok(n, K, N) || !dtype_ok(dtype) ||
      (scale != nullptr && (opt->block == 32 || !ok_ptr(scale, false))))
    return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!ok_ptr(w, true) || !ok_ptr(codes, true) || !ok_ptr(scales, false))
    return MOE_ERR_INVALID_ARG;
  return status_of(MOE_MX_PICK(
      quantize_weights, (n, K, N, w, scale, codes, scales, stream)));
}

moe_status_t moe_mx_pack(const moe_mx_t* opt, int32_t n, int32_t K, int32_t N,
                         const uint8_t* codes, const uint8_t* scales,
                         void* packed, moe_stream_t stream) {
  if (!mx::options_ok(opt) || !matrix_ok(n, K, N)) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!ok_ptr(codes, true) || !ok_ptr(scales, false) || !ok_ptr(packed, true))
    return MOE_ERR_INVALID_ARG;
  const Layout l = {K, N, opt->block};
  char* p = static_cast<char*>(packed);
  if (opt->block == 16)
    pack_kernel<16><<<record_grid(l, n), kThreads, 0, stream>>>(codes, scales,
                                                                n, l, p);
  else
    pack_kernel<32><<<record_grid(l, n), kThreads, 0, stream>>>(codes, scales,
                                                                n, l, p);
  return launched();
}

moe_status_t moe_mx_dequantize(const moe_mx_t* opt, int32_t n, int32_t K,
                               int32_t N, const void* packed,
                               const float* scale, moe_dtype_t dtype, void* w,
                               moe_stream_t stream) {
  if (!mx::options_ok(opt) || !matrix_ok(n, K, N) || !dtype_ok(dtype) ||
      (scale != nullptr && (opt->block == 32 || !ok_ptr(scale, false))))
    return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!ok_ptr(packed, true) || !ok_ptr(w, true)) return MOE_ERR_INVALID_ARG;
  const Layout l = {K, N, opt->block};
  const char* p = static_cast<const char*>(packed);
  const dim3 grid = record_grid(l, n);
#define MOE_MX_EXPAND(B, T)                                               \
  dequantize_kernel<B, T><<<grid, kThreads, 0, stream>>>(p, scale, n, l, \
                                                         static_cast<T*>(w))
  if (opt->block == 16) {
    if (dtype == MOE_F32)
      MOE_MX_EXPAND(16, float);
    else
      MOE_MX_EXPAND(16, __nv_bfloat16);
  } else if (dtype == MOE_F32) {
    MOE_MX_EXPAND(32, float);
  } else {
    MOE_MX_EXPAND(32, __nv_bfloat16);
  }
#undef MOE_MX_EXPAND
  return launched();
}

}  // extern "C"
