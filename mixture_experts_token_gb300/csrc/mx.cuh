// Microscaled 4-bit floating point (internal): the number formats, a block's
// scale and codes, and the layout of weight matrices.
//
// A code is a sign, two exponent bits and a mantissa bit: 0, 0.5, 1, 1.5, 2,
// 3, 4, 6.  Blocks of 32 along the reduction axis share a power of two (the
// biased exponent in a byte, 255 for NaN), blocks of 16 a number of 4 exponent
// and 3 mantissa bits (0x7f for NaN) under a float32 scale of the tensor.
// Rows of codes: K/2 bytes, column 2i in the low four bits of byte i; rows of
// scales of a weight matrix: scale_row() bytes, one a block, zeros behind the
// last.  The scales of the products' rows lie by 256 of K: for each of those,
// for each row, its 256 / block, so that what a product wants of 32 rows at a
// time lies together.
//
// A packed matrix [K, N] is, for each tile of 128 columns, one record after
// another, a record for each 256 of K:
//   codes   128 rows (columns of the matrix) of 128 bytes, 16-byte pieces
//           exchanged as the tensor cores' 128-byte swizzle has it (piece p of
//           row r lies at p ^ (r & 7))
//   scales  tiles of 512 bytes, each 4 scales of 128 rows: those of row r are
//           the word at (r % 32) * 16 + r / 32 * 4, the order in which 32 lanes
//           of tensor memory take four columns
// so that a product brings a record with one bulk copy and uses it in place.
// What lies past the matrix has code 0 and scale 0.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace moe {
namespace mx {

constexpr int kStageK = 256;
constexpr int kTileN = 128;
constexpr int kCodeBytes = kTileN * kStageK / 2;
constexpr int kScaleTile = 512;  // bytes: 4 scales of each of 128 rows
constexpr float kCodeMax = 6.0f;

__host__ __device__ constexpr int scale_tiles(int block) {  // of a record
  return kStageK / block / 4;
}
__host__ __device__ constexpr int record_bytes(int block) {
  return kCodeBytes + kScaleTile * scale_tiles(block);
}
__host__ __device__ inline int scale_row(int K, int block) {
  return (K / block + 3) / 4 * 4;
}

// Where the scale of block `at` of a row is, of R rows.
__host__ __device__ inline long long row_scale_at(int block, long long R,
                                                  long long row, int at) {
  const int per = kStageK / block;
  return (at / per * R + row) * per + at % per;
}
__host__ __device__ inline long long row_scale_bytes(int block, long long R,
                                                     int K) {
  return (K + kStageK - 1) / kStageK * R * (kStageK / block);
}

struct Layout {
  int K, N, block;
  __host__ __device__ int stages() const {
    return (K + kStageK - 1) / kStageK;
  }
  __host__ __device__ int tiles_n() const {
    return (N + kTileN - 1) / kTileN;
  }
  __host__ __device__ long long tile() const {
    return static_cast<long long>(stages()) * record_bytes(block);
  }
  __host__ __device__ long long matrix() const { return tile() * tiles_n(); }
};

inline bool scale_ok(int block, float s) {
  return block == 32 ? s == 1.0f : s >= 1.17549435e-38f && s <= 1e38f;
}
inline bool options_ok(const moe_mx_t* o) {
  return o != nullptr && (o->block == 16 || o->block == 32) &&
         scale_ok(o->block, o->x_scale) && scale_ok(o->block, o->h_scale);
}
// Blocks do not straddle rows, and rows of codes are whole 16-byte pieces.
inline bool length_ok(int K) {
  return K >= 32 && K % 32 == 0 && K <= (1 << 20);
}

// ---------------------------------------------------------- numbers ------
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16(v);
}

// Eight codes, the first in the lowest four bits: nearest, ties to the even
// code, magnitudes over 6 to 6.
__device__ __forceinline__ uint32_t encode8(const float (&q)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}\n"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]),
        "f"(q[6]), "f"(q[7]));
  return r;
}
// The values of eight codes.
__device__ __forceinline__ void decode8(uint32_t codes, float (&v)[8]) {
  uint32_t h[4];  // pairs of halves, exactly
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
// The value of a block's scale.
template <int BLOCK>
__device__ __forceinline__ float scale_value(uint32_t byte) {
  if (BLOCK == 32)
    return byte == 255   ? __uint_as_float(0x7fc00000u)
           : byte == 0 ? __uint_as_float(0x00400000u)  // 2^-127
                       : __uint_as_float(byte << 23);
  const uint32_t m = byte & 7, e = byte >> 3 & 15;
  if ((byte & 127) == 127) return __uint_as_float(0x7fc00000u);
  return e == 0 ? static_cast<float>(m) * 0.001953125f  // 2^-9
                : __uint_as_float((e + 120) << 23 | m << 20);
}

// A block's scale from the largest magnitude in it, as a float's bits (those
// of an infinity or a NaN are the largest): the scale's byte, and what its
// values are multiplied by (`inv`, and for blocks of 16 the scale `s`, with
// which the quotient is corrected).
struct Block {
  uint32_t byte;
  float s, inv;
};
template <int BLOCK>
__device__ __forceinline__ Block block_scale(uint32_t most) {
  Block b;
  if (BLOCK == 32) {
    // 2^(floor(log2 most) - 2): with the exponents' bias, the field less 2
    const uint32_t e = most >> 23;
    b.byte = e == 255 ? 255u : e > 2 ? e - 2 : 0u;
    b.s = 0.0f;
    b.inv = __uint_as_float((254u - min(b.byte, 253u)) << 23);
  } else {
    // The quotient by 6 and the reciprocal, each an approximation and one
    // Newton step: the nearest float but for an ulp at most, and m / 6 exact
    // where it is the middle of two scales (as a middle of two codes below).
    const bool finite = most < 0x7f800000u;
    const float m = __uint_as_float(most), q = m * (1.0f / kCodeMax);
    const float sixth = fmaf(fmaf(-q, kCodeMax, m), 1.0f / kCodeMax, q);
    uint32_t r, h;
    asm("{\n\t.reg .b16 t;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 t, %2, %3;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, t;\n\t"
        "cvt.u32.u16 %0, t;\n\t}\n"
        : "=r"(r), "=r"(h)
        : "f"(0.0f), "f"(finite ? sixth : 0.0f));
    b.byte = finite ? r : 127u;
    b.s = __low2float(*reinterpret_cast<const __half2*>(&h));
    float inv;
    asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(b.s));
    b.inv = b.s > 0.0f ? fmaf(fmaf(-b.s, inv, 1.0f), inv, inv) : 0.0f;
  }
  return b;
}
// v over the scale.  For blocks of 16 one step of correction makes the
// quotient the nearest float: v = m s for a midpoint m between two codes must
// give m itself, which the product with the reciprocal alone may miss.  (No
// other v gives m: v and m s, of at most 7 bits, differ by more than half an
// ulp of the quotient.)  Written so that a zero keeps its sign.
template <int BLOCK>
__device__ __forceinline__ float over_scale(float v, const Block& b) {
  const float q = v * b.inv;
  return BLOCK == 32 ? q : fmaf(-fmaf(q, b.s, -v), b.inv, q);
}

// Two numbers an instruction: quantising is bound by the instructions issued.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const unsigned long long*>(&a)),
        "l"(*reinterpret_cast<const unsigned long long*>(&b)));
  return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const unsigned long long*>(&a)),
        "l"(*reinterpret_cast<const unsigned long long*>(&b)),
        "l"(*reinterpret_cast<const unsigned long long*>(&c)));
  return *reinterpret_cast<const float2*>(&d);
}
// over_scale() of r v for two v, each with a block (r: 1 with blocks of 32), in
// the same steps with the signs of v, the reciprocal and the remainder turned.
template <int BLOCK>
__device__ __forceinline__ float2 over_scale2(float2 v, float r,
                                              const Block& b,
                                              const Block& c) {
  if (BLOCK == 32) return mul2(v, make_float2(b.inv, c.inv));
  const float2 inv = make_float2(-b.inv, -c.inv);
  const float2 minus = mul2(v, make_float2(-r, -r)), q = mul2(minus, inv);
  return fma2(fma2(q, make_float2(b.s, c.s), minus), inv, q);
}

// Magnitudes, as bits whose order is theirs; those of a NaN or an infinity are
// larger than any number's.
__device__ __forceinline__ uint32_t largest(const float (&v)[8]) {
  uint32_t most = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    most = max(most, __float_as_uint(v[j]) & 0x7fffffffu);
  return most;
}
// of pairs of bf16 numbers: those of the pairs' low halves and high halves
__device__ __forceinline__ uint32_t largest2(uint32_t most, uint32_t pair) {
  const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162*>(&most);
  const uint32_t mag = pair & 0x7fff7fffu;
  const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&mag);
  const __nv_bfloat162 m = __hmax2_nan(a, b);
  return *reinterpret_cast<const uint32_t*>(&m);
}
// The largest magnitude of values that are multiplied by r, from that of the
// values: rounding keeps order.
__device__ __forceinline__ uint32_t scaled_bits(uint32_t most, float r) {
  return __float_as_uint(__uint_as_float(most) * r) & 0x7fffffffu;
}

}  // namespace mx
}  // namespace moe
