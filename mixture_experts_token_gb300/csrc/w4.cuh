// Layout of 4-bit weight matrices (internal).  A matrix [K, N] of one expert
// is stored as ceil(N / 16) records of 16 columns, one after another:
//
//   for each step of 256 rows of K (the last may have fewer tiles):
//     codes   tiles of 64 x 16 codes, 512 bytes each
//     scales  [8][256 / group] pairs of bf16: (column c, column c + 8) of the
//             step's group g at [c][g]
//     zeros   the same with pairs of bytes (only with zero points)
//
// so that a product copies one contiguous piece a step.  A tile is one 16-byte
// load per lane of a warp.  Word s of the lane is the weight operand of one
// m16n8k16 matrix instruction, rows 16 s to 16 s + 15 of the tile: with
// c = lane / 4, t = lane % 4 and k = 16 s + 2 t its nibbles, low to high, are
//   (c,k) (c+8,k) (c,k+8) (c+8,k+8) (c,k+1) (c+8,k+1) (c,k+9) (c+8,k+9)
// so that masking two nibbles 16 bits apart yields a packed operand pair.
// Two words never mix groups of 32 rows.  Codes of rows and columns past the
// matrix are the zero point, so they weigh nothing.
#pragma once

#include "internal.h"

namespace moe {
namespace w4 {

constexpr int kTileK = 64;
constexpr int kTileN = 16;
constexpr int kTileBytes = kTileK * kTileN / 2;
constexpr int kStepK = 256;  // rows of a step: four tiles

struct Layout {
  int K, N, group;
  bool zeros;
  __host__ __device__ int tiles_k() const {
    return (K + kTileK - 1) / kTileK;
  }
  __host__ __device__ int tiles_n() const {
    return (N + kTileN - 1) / kTileN;
  }
  __host__ __device__ int groups() const { return (K + group - 1) / group; }
  __host__ __device__ int steps() const { return (K + kStepK - 1) / kStepK; }
  __host__ __device__ int scale_bytes() const {  // scales and zeros of a step
    return 8 * (kStepK / group) * (zeros ? 6 : 4);
  }
  // Bytes from a record's start to a step, and to its scales.
  __host__ __device__ long long step_at(int s) const {
    return static_cast<long long>(s) *
           (kStepK / kTileK * kTileBytes + scale_bytes());
  }
  __host__ __device__ long long scales_at(int s) const {
    const int left = tiles_k() - s * (kStepK / kTileK);
    return step_at(s) +
           (left < kStepK / kTileK ? left : kStepK / kTileK) * kTileBytes;
  }
  __host__ __device__ long long record() const {
    return scales_at(steps() - 1) + scale_bytes();
  }
  __host__ __device__ long long matrix() const { return record() * tiles_n(); }
};

inline bool options_ok(const moe_w4_t* o) {
  return o != nullptr &&
         (o->group_size == 32 || o->group_size == 64 ||
          o->group_size == 128) &&
         (o->zero_points == 0 || o->zero_points == 1);
}
inline Layout layout(const moe_w4_t& o, int K, int N) {
  return {K, N, o.group_size, o.zero_points != 0};
}

}  // namespace w4
}  // namespace moe
