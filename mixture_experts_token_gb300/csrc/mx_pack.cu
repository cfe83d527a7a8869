// Microscaled 4-bit numbers (mx.cuh): quantising rows and weight matrices,
// laying matrices out for the products, and expanding both again.  Each
// kernel reads its input once and writes its output once.  Measured: 8192 x
// 7168 bf16 rows, blocks of 32, quantised 28 to 31 us, expanded 23 to 24 (148 MB
// each, 22 us at 6.8 TB/s); eight bf16 matrices of 7168 x 2048, blocks of 16,
// quantised 67 us (301 MB, 44 us), packed 22 (132 MB, 19), expanded 48 (301 MB,
// 44).  Rows both ways and quantising matrices are bound by issue (slots 64 to 77%
// busy), the others by bytes.
#include "launch.cuh"
#include "mx.cuh"

namespace moe {
namespace {

using namespace mx;

constexpr int kThreads = 256;

// Eight values as they lie in memory.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  }
  __device__ __forceinline__ uint32_t most() const { return largest(v); }
  __device__ __forceinline__ float at(int j) const { return v[j]; }
};
template <>
struct Eight<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
  __device__ __forceinline__ uint32_t most() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = largest2(m, w[i]);
    return max(m << 16, m & 0xffff0000u);
  }
  __device__ __forceinline__ float at(int j) const {
    return __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
  }
};
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

// Rows, eight values a thread and a piece; a CTA takes kPieces * kThreads
// pieces in a row, all of which it loads before it uses one.  (Plain loads:
// those of constant memory may not see what the kernel before writes while
// this one has begun.)
constexpr int kPieces = 4;

// The row and the place in it of a thread's pieces, kThreads apart.
struct Place {
  long long row;
  uint32_t at, per_row;
  __device__ __forceinline__ Place(long long first, int per_row)
      : row(first / per_row), per_row(per_row) {
    at = static_cast<uint32_t>(first - row * per_row) + threadIdx.x;
    wrap();
  }
  __device__ __forceinline__ void next() {
    at += kThreads;
    if (per_row >= kThreads) {
      if (at >= per_row) {
        at -= per_row;
        ++row;
      }
    } else {
      wrap();
    }
  }
  __device__ __forceinline__ void wrap() {
    const uint32_t down = at / per_row;
    row += down;
    at -= down * per_row;
  }
};

// A block is two or four lanes.
template <int BLOCK, typename T>
__global__ void __launch_bounds__(kThreads)
    quantize_rows_kernel(const T* x, int R, int K, float r, uint8_t* codes,
                         uint8_t* scales) {
  constexpr int kLanes = BLOCK / 8;
  launch::wait_for_previous();
  launch::let_next_start();
  const long long pieces = static_cast<long long>(R) * (K / 8);
  const long long first =
      blockIdx.x * static_cast<long long>(kPieces * kThreads);
  const bool all = first + kPieces * kThreads <= pieces;
  Place place(first, K / 8);
  Eight<T> v[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const long long i = first + p * kThreads + threadIdx.x;
    if (all || i < pieces)
      v[p].load(x + i * 8);
    else
      v[p].zero();
  }
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const long long i = first + p * kThreads + threadIdx.x;
    uint32_t most = v[p].most();
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1)
      most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    const Block b =
        block_scale<BLOCK>(BLOCK == 16 ? scaled_bits(most, r) : most);
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 two = over_scale2<BLOCK>(
          make_float2(v[p].at(j), v[p].at(j + 1)), r, b, b);
      q[j] = two.x;
      q[j + 1] = two.y;
    }
    const uint32_t c = encode8(q);
    if (all || i < pieces) {
      reinterpret_cast<uint32_t*>(codes)[i] = c;
      if (threadIdx.x % kLanes == 0) {
        const int at = static_cast<int>(place.at) / kLanes;
        uint8_t* s = scales + row_scale_at(BLOCK, R, place.row, at);
        *s = static_cast<uint8_t>(b.byte);
        if (at == K / BLOCK - 1)  // zeros to the end of the 256
          for (int j = at + 1; j % (kStageK / BLOCK) != 0; ++j) *++s = 0;
      }
    }
    place.next();
  }
}

template <int BLOCK, typename T>
__global__ void __launch_bounds__(kThreads)
    dequantize_rows_kernel(const uint8_t* codes, const uint8_t* scales, int R,
                           int K, float scale, T* x) {
  launch::wait_for_previous();
  launch::let_next_start();
  const long long pieces = static_cast<long long>(R) * (K / 8);
  const long long first =
      blockIdx.x * static_cast<long long>(kPieces * kThreads);
  Place place(first, K / 8);
  uint32_t c[kPieces], byte[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const long long i = first + p * kThreads + threadIdx.x;
    if (i < pieces) {
      c[p] = reinterpret_cast<const uint32_t*>(codes)[i];
      byte[p] = scales[row_scale_at(BLOCK, R, place.row,
                                    place.at / (BLOCK / 8))];
    }
    place.next();
  }
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const long long i = first + p * kThreads + threadIdx.x;
    if (i >= pieces) return;
    const float s = scale_value<BLOCK>(byte[p]);
    float v[8];
    decode8(c[p], v);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float2 two = mul2(make_float2(v[j], v[j + 1]), make_float2(s, s));  // exact
      if (BLOCK == 16) two = mul2(two, make_float2(scale, scale));
      v[j] = two.x;
      v[j + 1] = two.y;
    }
    store8(v, x + i * 8);
  }
}

// A weight matrix w [K, N] becomes N rows of codes: 64 columns and 256 of K at
// a time through shared memory, read a row of w and written a row of codes at
// a time.  A warp has 32 of K, a lane two neighbouring columns of them.  (What a
// thread loads at once passes its registers: blocks of 16 and 32 spill 16 and 52
// bytes in bf16, under 64 registers, 144 and 248 in float32, under 80.)
constexpr int kTurnN = 64;
template <typename T>
struct Two;
template <>
struct Two<float> {
  uint32_t m[2] = {0, 0};  // the largest magnitudes so far
  static __device__ __forceinline__ float2 load(const float* p) {
    return *reinterpret_cast<const float2*>(p);
  }
  __device__ __forceinline__ void look(const float* p) {
    const uint2 f = *reinterpret_cast<const uint2*>(p);
    m[0] = max(m[0], f.x & 0x7fffffffu);
    m[1] = max(m[1], f.y & 0x7fffffffu);
  }
  __device__ __forceinline__ uint32_t most(int n) const { return m[n]; }
};
template <>
struct Two<__nv_bfloat16> {
  uint32_t m = 0;
  static __device__ __forceinline__ float2 load(const __nv_bfloat16* p) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
  }
  __device__ __forceinline__ void look(const __nv_bfloat16* p) {
    m = largest2(m, *reinterpret_cast<const uint32_t*>(p));
  }
  __device__ __forceinline__ uint32_t most(int n) const {
    return n ? m & 0xffff0000u : m << 16;
  }
};

template <int BLOCK, typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3)
    quantize_weights_kernel(const T* __restrict__ w,
                            const float* __restrict__ scale, int n_mats,
                            int K, int N, uint8_t* __restrict__ codes,
                            uint8_t* __restrict__ scales) {
  constexpr int kPer = 16 / sizeof(T);  // values of a 16-byte piece
  constexpr int kRow = kStageK / BLOCK;  // scales of a row here
  static_assert(kThreads / 32 * 32 == kStageK, "a warp has 32 of K");
  extern __shared__ __align__(16) char raw[];
  T* tile = reinterpret_cast<T*>(raw);  // [256][64]
  __shared__ __align__(16) char out[kTurnN * kStageK / 2];
  __shared__ __align__(4) uint8_t out_s[kTurnN][kRow];
  const int n0 = blockIdx.x * kTurnN, k0 = blockIdx.y * kStageK;
  const int sr = scale_row(K, BLOCK);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k_here = min(kStageK, K - k0), n_here = min(kTurnN, N - n0);
  // whole pieces, each in bounds and aligned
  const bool wide = N % kPer == 0;
  for (long long m = blockIdx.z; m < n_mats; m += gridDim.z) {
    const float r = BLOCK == 16 && scale ? __frcp_rn(scale[m]) : 1.0f;
    const T* src = w + (m * K + k0) * N + n0;
    __syncthreads();
    if (wide) {
      constexpr int kIn = kStageK * kTurnN / kPer / kThreads;
      uint4 v[kIn];
#pragma unroll
      for (int i = 0; i < kIn; ++i) {
        const int at = i * kThreads + threadIdx.x;
        const int k = at / (kTurnN / kPer), n = at % (kTurnN / kPer) * kPer;
        if (k < k_here && n < n_here)
          v[i] = __ldg(reinterpret_cast<const uint4*>(
              src + static_cast<long long>(k) * N + n));
      }
#pragma unroll
      for (int i = 0; i < kIn; ++i)
        reinterpret_cast<uint4*>(raw)[i * kThreads + threadIdx.x] = v[i];
    } else {
      for (int i = threadIdx.x; i < kStageK * kTurnN; i += kThreads) {
        const int k = i / kTurnN, n = i % kTurnN;
        if (k < k_here && n < n_here)
          tile[i] = src[static_cast<long long>(k) * N + n];
      }
    }
    __syncthreads();
    if (warp * 32 < k_here) {  // K is a multiple of 32
      uint32_t c[2][4];
      const T* col = tile + warp * 32 * kTurnN + 2 * lane;
#pragma unroll
      for (int h = 0; h < 32 / BLOCK; ++h) {
        // read twice: held in registers, the values would cost warps
        Two<T> two;
#pragma unroll
        for (int j = 0; j < BLOCK; ++j)
          two.look(col + (h * BLOCK + j) * kTurnN);
        Block b[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          b[n] = block_scale<BLOCK>(BLOCK == 16 ? scaled_bits(two.most(n), r)
                                                : two.most(n));
          out_s[2 * lane + n][warp * (32 / BLOCK) + h] =
              static_cast<uint8_t>(b[n].byte);
        }
#pragma unroll
        for (int j = 0; j < BLOCK / 8; ++j) {
          float q[2][8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 f = over_scale2<BLOCK>(
                Two<T>::load(col + (h * BLOCK + 8 * j + e) * kTurnN), r, b[0],
                b[1]);
            q[0][e] = f.x;
            q[1][e] = f.y;
          }
          c[0][h * (BLOCK / 8) + j] = encode8(q[0]);
          c[1][h * (BLOCK / 8) + j] = encode8(q[1]);
        }
      }
      // pieces of a row change places by the row, so that lanes meet no bank
#pragma unroll
      for (int n = 0; n < 2; ++n)
        *reinterpret_cast<uint4*>(out + (2 * lane + n) * (kStageK / 2) +
                                  ((warp ^ (lane & 7)) << 4)) =
            make_uint4(c[n][0], c[n][1], c[n][2], c[n][3]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kTurnN * 8; i += kThreads) {
      const int n = i / 8, p = i % 8;
      if (n < n_here && p * 32 < k_here)
        *reinterpret_cast<uint4*>(codes + (m * N + n0 + n) * (K / 2) +
                                  k0 / 2 + p * 16) =
            *reinterpret_cast<const uint4*>(out + n * (kStageK / 2) +
                                            ((p ^ (n >> 1 & 7)) << 4));
    }
    const int words = min(kRow, sr - k0 / BLOCK) / 4;  // zeros behind the last
    for (int i = threadIdx.x; i < kTurnN * words; i += kThreads) {
      const int n = i / words, at = i % words * 4;
      uint32_t v = *reinterpret_cast<const uint32_t*>(&out_s[n][at]);
      const int left = k_here / BLOCK - at;
      if (left < 4) v &= (1u << (8 * left)) - 1;
      if (n < n_here)
        *reinterpret_cast<uint32_t*>(scales + (m * N + n0 + n) * sr +
                                     k0 / BLOCK + at) = v;
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

__device__ __forceinline__ void store2(float2 v, float* p) {
  *reinterpret_cast<float2*>(p) = v;
}
__device__ __forceinline__ void store2(float2 v, __nv_bfloat16* p) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}

// Records to w [K, N], a CTA for each: a thread expands 32 of K of two
// neighbouring columns, and a warp writes 64 columns of a row side by side.
template <int BLOCK, typename T>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const char* __restrict__ packed,
                      const float* __restrict__ scale, int n_mats, Layout l,
                      T* __restrict__ w) {
  __shared__ __align__(16) char rec[record_bytes(BLOCK)];
  const int stage = blockIdx.x, n0 = blockIdx.y * kTileN;
  const bool pairs = l.N % 2 == 0;
  for (long long m = blockIdx.z; m < n_mats; m += gridDim.z) {
    const char* src = packed + m * l.matrix() + blockIdx.y * l.tile() +
                      static_cast<long long>(stage) * record_bytes(BLOCK);
    __syncthreads();
    for (int i = threadIdx.x; i < record_bytes(BLOCK) / 16; i += kThreads)
      reinterpret_cast<uint4*>(rec)[i] =
          __ldg(reinterpret_cast<const uint4*>(src) + i);
    __syncthreads();
    const float t = BLOCK == 16 && scale ? scale[m] : 1.0f;
    for (int i = threadIdx.x; i < kTileN / 2 * 8; i += kThreads) {
      const int r = i % (kTileN / 2) * 2, p = i / (kTileN / 2);
      const int k = stage * kStageK + p * 32;
      if (n0 + r >= l.N || k >= l.K) continue;
      uint32_t c[2][4];
      float s[2][32 / BLOCK];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int row = r + n;
        const uint4 v = *reinterpret_cast<const uint4*>(
            rec + row * 128 + ((p ^ (row & 7)) << 4));
        c[n][0] = v.x, c[n][1] = v.y, c[n][2] = v.z, c[n][3] = v.w;
#pragma unroll
        for (int h = 0; h < 32 / BLOCK; ++h) {
          const int g = p * (32 / BLOCK) + h;
          s[n][h] = scale_value<BLOCK>(static_cast<uint8_t>(
              rec[kCodeBytes + g / 4 * kScaleTile + row % 32 * 16 +
                  row / 32 * 4 + g % 4]));
        }
      }
      T* out = w + (m * l.K + k) * l.N + n0 + r;
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        float v[2][8];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          decode8(c[n][j / 8], v[n]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[n][i] *= s[n][j / BLOCK];
            if (BLOCK == 16) v[n][i] *= t;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i, out += l.N) {
          if (pairs) {
            store2(make_float2(v[0][i], v[1][i]), out);
          } else {
            put(out, v[0][i]);
            if (n0 + r + 1 < l.N) put(out + 1, v[1][i]);
          }
        }
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
// What a grid holds, about 10^13 values: more than any memory does.
bool grid_ok(long long pieces) {
  return pieces <= static_cast<long long>(kPieces * kThreads) * 0x7fffffff;
}
unsigned row_grid(long long pieces) {
  return static_cast<unsigned>((pieces + kPieces * kThreads - 1) /
                               (kPieces * kThreads));
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
  const int bytes = kStageK * kTurnN * sizeof(T);
  kernel<<<grid, kThreads, bytes, s>>>(static_cast<const T*>(w), scale, n, K,
                                       N, codes, scales);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_rows(int block, int R, int K, moe_dtype_t dtype,
                           const void* x, float scale, uint8_t* codes,
                           uint8_t* scales, cudaStream_t s) {
  const long long pieces = static_cast<long long>(R) * (K / 8);
  if (!grid_ok(pieces)) return cudaErrorInvalidValue;
  const float r = 1.0f / scale;
  const unsigned grid = row_grid(pieces);
#define MOE_MX_ROWS(B, T)                                                   \
  return launch::overlapping(quantize_rows_kernel<B, T>, grid, kThreads, 0, \
                             s, static_cast<const T*>(x), R, K, r,          \
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
  const size_t each = static_cast<size_t>(Layout{K, N, opt->block}.matrix());
  if (n > 0 && each > SIZE_MAX / n) return 0;  // no such number of bytes
  return each * n;
}

size_t moe_mx_row_scale_bytes(const moe_mx_t* opt, int32_t R, int32_t K) {
  if (!mx::options_ok(opt) || !rows_ok(R, K)) return 0;
  return static_cast<size_t>(row_scale_bytes(opt->block, R, K));
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
  if (!ok_ptr(x, true) || !ok_ptr(codes, true) || !ok_ptr(scales, true))
    return MOE_ERR_INVALID_ARG;
  if (!grid_ok(static_cast<long long>(R) * (K / 8)))
    return MOE_ERR_UNSUPPORTED;
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
  if (!ok_ptr(codes, true) || !ok_ptr(scales, true) || !ok_ptr(x, true))
    return MOE_ERR_INVALID_ARG;
  const long long pieces = static_cast<long long>(R) * (K / 8);
  if (!grid_ok(pieces)) return MOE_ERR_UNSUPPORTED;
  cudaError_t e;
#define MOE_MX_ROWS(B, T)                                             \
  e = launch::overlapping(dequantize_rows_kernel<B, T>, row_grid(pieces), \
                          kThreads, 0, stream, codes, scales, R, K, scale, \
                          static_cast<T*>(x))
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
  return status_of(e);
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
